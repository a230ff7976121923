// Pages with reference counts (kk_pages.cu).
#pragma once
#include "kk_internal.h"

namespace kk {

constexpr int kMaxPageArrays = 8;

struct PageArray {
  char* base;
  long long slice, page, bytes;  // strides and size in bytes
  int slices, vec;               // vec: bytes of a load, 16 or 4
  int per, vecs;                 // vectors of a slice, of a page
  int step_s, step_o;            // slices and vectors a thread moves on by from one of its vectors to the next
  int first;                     // chunks of the arrays before
  bool whole;                    // slices are whole chunks
};
struct PageArrays {
  PageArray a[kMaxPageArrays];
  int n;
  int chunks;  // of one page of every array
};
struct ForkArgs {
  Table bt;
  int bs, F, keep, num_pages;
  const int* parent;
  const int* refs_in;
  int* refs_out;
  int *child_pages, *child_offsets, *child_lens;
  int *kids, *first;  // [R]: children, the first of them
  int* at;            // [F + 1] where a child's copy is in the list
  int2* pairs;        // copies: from, to
  int* n_pairs;
  int* err;
};
struct CompactArgs {
  int num_pages;
  const int* refs_in;
  int* refs_out;
  const int* pages_in;
  int* pages_out;
  long long n;
  int *remap, *used;
  int2* pairs;
  int* n_pairs;
  int* err;
};
bool plan_page_arrays(PageArrays* pa);  // fills vec and what follows; false: too large
cudaError_t launch_pages_alloc(const int* refs_in, int* refs_out, int num_pages, const int* want, int n, int* out,
                               int* err, cudaStream_t s);
cudaError_t launch_pages_free(const Table& bt, const int* refs_in, int* refs_out, int num_pages, int* err,
                              cudaStream_t s);
cudaError_t launch_pages_fork(const ForkArgs& f, const PageArrays& pa, cudaStream_t s);
cudaError_t launch_pages_compact(const CompactArgs& c, const PageArrays& pa, cudaStream_t s);

}  // namespace kk
