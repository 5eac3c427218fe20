// Items dealt to the blocks of a grid in runs of equal length, the first blocks
// one more where they do not divide.  No product passes the number of items.
#pragma once
#ifdef __CUDACC__
#define MXFP8_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MXFP8_HOST_DEVICE inline
#endif

namespace mxfp8 {

struct EvenShare {
  int first, last;  // [first, last)
};
MXFP8_HOST_DEVICE EvenShare even_share(int items, int block, int blocks) {
  const int each = items / blocks, more = items % blocks;
  const int first = block * each + (block < more ? block : more);
  return {first, first + each + (block < more ? 1 : 0)};
}

}  // namespace mxfp8
