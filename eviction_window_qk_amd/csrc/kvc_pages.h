// Page tables: declarations shared by their kernels and host code.
#pragma once

#include "kvc_internal.h"

namespace kvc {

constexpr int kPageTile = 4096;     // pages a workgroup ranks
constexpr int kMaxBuffers = 16;     // buffers per launch (by value in the arguments)
constexpr int64_t kCopyChunk = 8192;  // bytes of a page one workgroup copies at a time

struct Pages {
  int B, tb, bs, n;  // sequences, entries each, positions per page, pages
  int32_t* table;
  int32_t* seq_len;
  int32_t* refs;
};

// Buffers of one launch; chunks of all of them are numbered through.
struct Buffers {
  int n;
  uint32_t chunks;  // per page, over all buffers
  struct {
    char* base;
    int64_t bytes;
    uint32_t first, unit;  // first chunk; widest power of two to 16 that divides base and bytes
  } b[kMaxBuffers];
};

// Workspace carve-up, in int32 elements.
struct PagesWs {
  size_t meta, count, list, movers, place, need, offset, kind, rank, from, total;
};
PagesWs pages_ws(const Pages& t, int n_pairs);

hipError_t launch_pages_alloc(const Pages& t, const int32_t* want, int32_t* status, int32_t* ws,
                              hipStream_t s);
// One launch per group of buffers; the first also writes the tables.
hipError_t launch_pages_fork(const Pages& t, int n_pairs, const int32_t* src, const int32_t* dst,
                             const Buffers* groups, int n_groups, int32_t* status, int32_t* ws,
                             hipStream_t s);
hipError_t launch_pages_free(const Pages& t, int n_ids, const int32_t* ids, hipStream_t s);
hipError_t launch_pages_copy(int n_blocks, int n_pairs, const int32_t* src, const int32_t* dst,
                             const Buffers* groups, int n_groups, hipStream_t s);
hipError_t launch_pages_compact(const Pages& t, const Buffers* groups, int n_groups,
                                int32_t* table_out, int32_t* refs_out, int32_t* remap,
                                int32_t* n_live, int32_t* ws, hipStream_t s);

}  // namespace kvc
